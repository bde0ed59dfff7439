// bf16 gradients of the feed-forward block (ffn_tiles.hpp): dh and dw2, which need
// nothing of each other, then dx and dw1, dw3, which need dh's dg and du.
#include "ffn_plan.hpp"

namespace moe {
namespace {

struct BackwardArgs {
  FfnTileArgs dh{}, dw2{}, dx{}, dw13{};
  BackwardArgs(const moe_ffn_t& f, const FfnTensors<uint16_t>& t) {
    dh.offsets = dw2.offsets = dx.offsets = dw13.offsets = t.offsets;
    dh.P0 = t.dy; dh.Q0 = t.w2; dh.cols = f.d_ff; dh.len = f.d_model;
    dh.g = t.g; dh.u = t.u; dh.o0 = t.dg; dh.o1 = t.du;
    dw2.P0 = t.dy; dw2.Q0 = t.h; dw2.rows = f.d_model; dw2.cols = f.d_ff; dw2.o0 = t.dw2;
    dx.P0 = t.dg; dx.P1 = t.du; dx.Q0 = t.w1; dx.Q1 = t.w3; dx.cols = f.d_model; dx.len = f.d_ff; dx.o0 = t.dx;
    dw13.P0 = t.dg; dw13.P1 = t.du; dw13.Q0 = t.x; dw13.rows = f.d_ff; dw13.cols = f.d_model;
    dw13.o0 = t.dw1; dw13.o1 = t.dw3;
  }
};

}  // namespace

size_t ffn_backward_product_bytes_bf16(const moe_ffn_t& f) {
  return std::max(FfnPairPlan::of(f, kDh, kDw2).workspace(), FfnPairPlan::of(f, kDx, kDw13).workspace());
}

hipError_t launch_ffn_backward_bf16(const moe_ffn_t& f, const FfnTensors<uint16_t>& t, void* partials, hipStream_t st) {
  const BackwardArgs a(f, t);
  const bool dx = t.dx != nullptr, dw13 = t.dw1 != nullptr, dw2 = t.dw2 != nullptr;
  if (!dx && !dw13) return launch_ffn_tiles<kDw2>(f, FfnPlans::of(f, kDw2), a.dw2, partials, st);
  const hipError_t e = dw2 ? launch_ffn_pair<kDh, kDw2>(f, FfnPairPlan::of(f, kDh, kDw2), a.dh, a.dw2, partials, st)
                           : launch_ffn_tiles<kDh>(f, FfnPlans::of(f, kDh), a.dh, partials, st);
  if (e != hipSuccess) return e;
  if (dx && dw13) return launch_ffn_pair<kDx, kDw13>(f, FfnPairPlan::of(f, kDx, kDw13), a.dx, a.dw13, partials, st);
  return dx ? launch_ffn_tiles<kDx>(f, FfnPlans::of(f, kDx), a.dx, partials, st)
            : launch_ffn_tiles<kDw13>(f, FfnPlans::of(f, kDw13), a.dw13, partials, st);
}

}  // namespace moe
