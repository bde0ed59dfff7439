// bf16 gradients of the feed-forward block from those at its pre-activations (ffn_tiles.hpp).
#include "ffn_plan.hpp"

namespace moe {

size_t ffn_backward_product_bytes_bf16(const moe_ffn_t& f) {
  size_t most = 0;
  for (int kind : {kDh, kDx, kDw13, kDw2}) most = std::max(most, FfnPlan::of(f, kind).workspace);
  return most;
}

hipError_t launch_ffn_backward_bf16(const moe_ffn_t& f, const FfnTensors<uint16_t>& t, void* partials, hipStream_t st) {
  hipError_t e = hipSuccess;
  FfnTileArgs a{};
  a.offsets = t.offsets;
  if (t.dw2 != nullptr) {
    a.P0 = t.dy; a.Q0 = t.h; a.rows = f.d_model; a.cols = f.d_ff; a.o0 = t.dw2;
    if ((e = launch_ffn_tiles<kDw2>(f, a, partials, st)) != hipSuccess) return e;
  }
  if (t.dx == nullptr && t.dw1 == nullptr) return e;
  if ((e = launch_ffn_dh_bf16(f, t, partials, st)) != hipSuccess) return e;
  a.P0 = t.dg; a.P1 = t.du;
  if (t.dx != nullptr) {
    a.Q0 = t.w1; a.Q1 = t.w3; a.cols = f.d_model; a.len = f.d_ff; a.o0 = t.dx;
    if ((e = launch_ffn_tiles<kDx>(f, a, partials, st)) != hipSuccess) return e;
  }
  if (t.dw1 == nullptr) return e;
  a.Q0 = t.x; a.Q1 = nullptr; a.rows = f.d_ff; a.cols = f.d_model; a.o0 = t.dw1; a.o1 = t.dw3;
  return launch_ffn_tiles<kDw13>(f, a, partials, st);
}

}  // namespace moe
