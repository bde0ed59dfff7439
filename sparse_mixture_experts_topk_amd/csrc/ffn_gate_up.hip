// bf16 gate/up product of the feed-forward block: up to kLinearDecodeRows rows of one
// group stream the weights (ffn_decode.hip); more, or few channels of a long
// contraction, run as tiles (ffn_tiles.hpp).
#include "ffn_plan.hpp"

namespace moe {
namespace {

struct GateUpPlan {
  bool stream = false;
  DecodeBlock block{};
  FfnPlans tiles{};

  static GateUpPlan of(const moe_ffn_t& f) {
    GateUpPlan p;
    const int cus = device_cu_count();
    double stream = 0;
    if (f.groups == 1 && f.M <= kLinearDecodeRows) {
      p.stream = true;
      // 8 channels of each weight make a block of 16
      const int eights = (f.d_ff + 7) / 8;
      if (eights * ((f.M + 3) / 4) <= cus) p.block = {4, 16};
      else if (eights * ((f.M + 7) / 8) <= cus) p.block = {8, 16};
      else if (f.M <= 16) p.block = {16, 16};
      else p.block = {32, eights > cus ? 32 : 16};
      if (eights > cus) return p;
      // (as for the dense product: a block of channels stays on one CU)
      stream = 2.0 * f.d_model * (p.block.channels + std::min(p.block.rows, f.M)) / kCuBytesPerUs;
      if (stream <= kTilesStart) return p;
    }
    p.tiles = FfnPlans::of(f, kGateUp);
    p.stream = p.stream && stream <= p.tiles.least().cost + kTilesStart;
    return p;
  }
};

}  // namespace

size_t ffn_gate_up_bytes_bf16(const moe_ffn_t& f) {
  const GateUpPlan p = GateUpPlan::of(f);
  return p.stream ? 0 : p.tiles.least().workspace;
}

hipError_t launch_ffn_gate_up_bf16(const moe_ffn_t& f, const FfnTensors<uint16_t>& t, void* workspace, hipStream_t st) {
  const GateUpPlan p = GateUpPlan::of(f);
  if (p.stream) return launch_ffn_decode(f, p.block, t, st);
  FfnTileArgs a{};
  a.P0 = t.x; a.Q0 = t.w1; a.Q1 = t.w3; a.offsets = t.offsets; a.cols = f.d_ff; a.len = f.d_model;
  a.o0 = t.h_out; a.o1 = t.g_out; a.o2 = t.u_out;
  return launch_ffn_tiles<kGateUp>(f, p.tiles, a, workspace, st);
}

}  // namespace moe
