// bf16 gate/up product of the feed-forward block, and the gradients at its pre-activations (ffn_tiles.hpp).
#include "ffn_plan.hpp"

namespace moe {

size_t ffn_gate_up_bytes_bf16(const moe_ffn_t& f) { return FfnPlan::of(f, kGateUp).workspace; }

hipError_t launch_ffn_gate_up_bf16(const moe_ffn_t& f, const FfnTensors<uint16_t>& t, void* workspace, hipStream_t st) {
  FfnTileArgs a{};
  a.P0 = t.x; a.Q0 = t.w1; a.Q1 = t.w3; a.offsets = t.offsets; a.cols = f.d_ff; a.len = f.d_model;
  a.o0 = t.h_out; a.o1 = t.g_out; a.o2 = t.u_out;
  return launch_ffn_tiles<kGateUp>(f, a, workspace, st);
}

hipError_t launch_ffn_dh_bf16(const moe_ffn_t& f, const FfnTensors<uint16_t>& t, void* partials, hipStream_t st) {
  FfnTileArgs a{};
  a.P0 = t.dy; a.Q0 = t.w2; a.offsets = t.offsets; a.cols = f.d_ff; a.len = f.d_model;
  a.g = t.g; a.u = t.u; a.o0 = t.dg; a.o1 = t.du;
  return launch_ffn_tiles<kDh>(f, a, partials, st);
}

}  // namespace moe
