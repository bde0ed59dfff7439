// Groups of rows of a feed-forward block (one per expert) and the four products on them.
#pragma once
#include "device_common.hpp"
#include "launch.hpp"

namespace moe {

// What a product computes.  g, u: the two pre-activations; every product sums over
// its contraction in fp32.
enum FfnKind {
  kGateUp,     // h = act(x w1^T) (x w3^T); g, u kept where asked for
  kDh,         // dh = dy w2, and from it dg = dh u act'(g), du = dh act(g)
  kDx,         // dg w1 + du w3
  kDw13,       // dg^T x and du^T x
  kDw2         // dy^T h
};
// Rows of these two are weights, and their contraction is over the rows of a group.
constexpr bool ffn_over_rows(int kind) { return kind == kDw13 || kind == kDw2; }

constexpr int kMaxFfnGroups = kMaxExpertGroups;

// Row offsets of the groups, in LDS: bounded to the buffers' rows and ascending,
// whatever the array holds (NULL: one group of all rows); and the tiles of
// `rows_per_tile` rows before each group.  By the first wavefront.
struct FfnGroups {
  int32_t off[kMaxFfnGroups + 1];
  int32_t pre[kMaxFfnGroups + 1];

  __device__ __forceinline__ void load(const int32_t* offsets, int groups, int M, int rows_per_tile) {
    if (threadIdx.x < kWave) {
      int carry = 0, high = 0;
      for (int base = 0; base <= groups; base += kWave) {
        const int e = base + (int)threadIdx.x;
        int o = 0;
        if (e <= groups) o = offsets != nullptr ? min(max(offsets[e], 0), M) : e == 0 ? 0 : M;
        // running maximum, then running tile count
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
          const int v = __shfl_up(o, d);
          if ((int)threadIdx.x >= d) o = max(o, v);
        }
        o = max(o, high);
        int before = __shfl_up(o, 1);
        if (threadIdx.x == 0) before = base == 0 ? o : high;
        int tiles = e == 0 ? 0 : (o - before + rows_per_tile - 1) / rows_per_tile;      // of group e - 1
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
          const int v = __shfl_up(tiles, d);
          if ((int)threadIdx.x >= d) tiles += v;
        }
        tiles += carry;
        if (e <= groups) {
          off[e] = o;
          pre[e] = tiles;
        }
        high = __shfl(o, kWave - 1);
        carry = __shfl(tiles, kWave - 1);
      }
    }
    __syncthreads();
  }
};

// A call's tensors; what it does not use is NULL.
template <class E>
struct FfnTensors {
  const int32_t* offsets;
  const E *x, *w1, *w3, *w2, *dy, *g, *u, *h;
  E *h_out, *g_out, *u_out;            // gate/up
  E *dx, *dw1, *dw3, *dw2;             // backward
  E *dg, *du;                          // backward: gradients at the pre-activations, in the workspace
};

// fp32 operands (ffn_f32.hip).
size_t ffn_gate_up_bytes_f32(const moe_ffn_t& f);
size_t ffn_backward_product_bytes_f32(const moe_ffn_t& f);
template <class E>
hipError_t launch_ffn_gate_up_f32(const moe_ffn_t& f, const FfnTensors<E>& t, void* workspace, hipStream_t st);
template <class E>
hipError_t launch_ffn_backward_f32(const moe_ffn_t& f, const FfnTensors<E>& t, void* partials, hipStream_t st);

}  // namespace moe
