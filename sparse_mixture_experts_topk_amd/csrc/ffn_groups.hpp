// Groups of rows of a feed-forward block (one per expert) and the four products on them.
#pragma once
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"

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
// whatever the array holds (NULL: one group of all rows); and running sums over the
// groups before each: of units(rows of the group), and of the groups that have rows.
struct FfnGroups {
  int32_t off[kMaxFfnGroups + 1];
  int32_t pre[kMaxFfnGroups + 1];
  int16_t full[kMaxFfnGroups + 1];

  // By the first wavefront; then a barrier.
  template <class Units>
  __device__ __forceinline__ void load(const int32_t* offsets, int groups, int M, Units&& units) {
    if (groups == 1) {
      if (threadIdx.x == 0) {
        off[0] = offsets != nullptr ? min(max(offsets[0], 0), M) : 0;
        off[1] = offsets != nullptr ? max(min(offsets[1], M), off[0]) : M;
        const int rows = off[1] - off[0];
        pre[0] = full[0] = 0;
        pre[1] = rows > 0 ? units(rows) : 0;
        full[1] = rows > 0;
      }
    } else if (threadIdx.x < kWave) {
      const int lane = threadIdx.x;
      int high = 0, carry = 0, count = 0;
      for (int base = 0; base <= groups; base += kWave) {
        const int e = base + lane;
        int o = 0;
        if (e <= groups) o = offsets != nullptr ? min(max(offsets[e], 0), M) : e == 0 ? 0 : M;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {                         // running maximum
          const int v = __shfl_up(o, d);
          if (lane >= d) o = max(o, v);
        }
        o = max(o, high);
        const int above = __shfl_up(o, 1), before = lane == 0 ? high : above;
        const bool there = e != 0 && e <= groups && o > before;       // group e - 1 has rows
        int sum = there ? units(o - before) : 0;
        const uint64_t rows = __ballot(there);
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
          const int v = __shfl_up(sum, d);
          if (lane >= d) sum += v;
        }
        sum += carry;
        if (e <= groups) {
          off[e] = o;
          pre[e] = sum;
          full[e] = (int16_t)(count + __popcll(rows & (~0ull >> (kWave - 1 - lane))));
        }
        high = __shfl(o, kWave - 1);
        carry = __shfl(sum, kWave - 1);
        count += __popcll(rows);
      }
    }
    __syncthreads();
  }
  // (uniform values)
  __device__ __forceinline__ int first(int e) const { return __builtin_amdgcn_readfirstlane(off[e]); }
  __device__ __forceinline__ int before(int e) const { return __builtin_amdgcn_readfirstlane(pre[e]); }
  __device__ __forceinline__ int full_before(int e) const { return __builtin_amdgcn_readfirstlane(full[e]); }
  // The last group with before(group) <= v: one that has units, if v is below their sum.
  __device__ __forceinline__ int of(int v, int groups) const {
    return last(groups, [&](int e) { return before(e) <= v; });
  }
  // The same for ascending v, from the last one's e.
  __device__ __forceinline__ int next(int e, int v, int groups) const {
    for (int i = 0; i < 2; ++i) {
      if (before(e + 1) > v) return e;
      ++e;
    }
    return before(e + 1) > v ? e : of(v, groups);
  }
  // The v-th of the groups that have rows.
  __device__ __forceinline__ int full_of(int v, int groups) const {
    return last(groups, [&](int e) { return full_before(e) <= v; });
  }
  // The v-th of those that have none.
  __device__ __forceinline__ int empty_of(int v, int groups) const {
    return last(groups, [&](int e) { return e - full_before(e) <= v; });
  }

 private:
  template <class Below>
  __device__ static __forceinline__ int last(int groups, Below&& below) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (below(mid)) lo = mid;
      else hi = mid;
    }
    return lo;
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

// bf16 operands: each call's products (ffn_gate_up.hip, ffn_gradients.hip).
size_t ffn_gate_up_bytes_bf16(const moe_ffn_t& f);
size_t ffn_backward_product_bytes_bf16(const moe_ffn_t& f);
hipError_t launch_ffn_gate_up_bf16(const moe_ffn_t& f, const FfnTensors<uint16_t>& t, void* workspace, hipStream_t st);
hipError_t launch_ffn_backward_bf16(const moe_ffn_t& f, const FfnTensors<uint16_t>& t, void* partials, hipStream_t st);

// ... gate/up of up to kLinearDecodeRows rows of one group with streamed weights (ffn_decode.hip).
hipError_t launch_ffn_decode(const moe_ffn_t& f, const DecodeBlock& b, const FfnTensors<uint16_t>& t, hipStream_t st);

// fp32 operands (ffn_f32.hip).
size_t ffn_gate_up_bytes_f32(const moe_ffn_t& f);
size_t ffn_backward_product_bytes_f32(const moe_ffn_t& f);
hipError_t launch_ffn_gate_up_f32(const moe_ffn_t& f, const FfnTensors<float>& t, void* workspace, hipStream_t st);
hipError_t launch_ffn_backward_f32(const moe_ffn_t& f, const FfnTensors<float>& t, void* partials, hipStream_t st);

}  // namespace moe
