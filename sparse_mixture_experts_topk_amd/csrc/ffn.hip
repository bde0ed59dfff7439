// Gated feed-forward block: gate/up forward and the gradients of the whole block.
//
// Pages: "Mixtral" study notes, MixtralExpert.forward = w2(silu(w1 x) * w3 x), differentiated:
//   dh = dy w2,  dg = dh u act'(g),  du = dh act(g)
//   dx = dg w1 + du w3,  dw1 = dg^T x,  dw3 = du^T x,  dw2 = dy^T h
#include <algorithm>

#include "ffn_groups.hpp"
#include "launch.hpp"

namespace moe {
namespace {

size_t elem(const moe_ffn_t& f) { return f.dtype == MOE_F32 ? 4 : 2; }
size_t pre_bytes(const moe_ffn_t& f) { return ((size_t)f.M * f.d_ff * elem(f) + 255) / 256 * 256; }

}  // namespace

size_t ffn_gate_up_workspace_bytes(const moe_ffn_t& f) {
  return f.dtype == MOE_F32 ? ffn_gate_up_bytes_f32(f) : ffn_gate_up_bytes_bf16(f);
}

size_t ffn_backward_workspace_bytes(const moe_ffn_t& f) {
  return 2 * pre_bytes(f) + (f.dtype == MOE_F32 ? ffn_backward_product_bytes_f32(f) : ffn_backward_product_bytes_bf16(f));
}

hipError_t launch_ffn_gate_up(const moe_ffn_t& f, const void* x, const int32_t* offsets, const void* w1,
                              const void* w3, void* h, void* pre1, void* pre3, void* workspace, hipStream_t st) {
  auto run = [&](auto e) {
    using E = decltype(e);
    FfnTensors<E> t{};
    t.offsets = offsets;
    t.x = static_cast<const E*>(x);
    t.w1 = static_cast<const E*>(w1);
    t.w3 = static_cast<const E*>(w3);
    t.h_out = static_cast<E*>(h);
    t.g_out = static_cast<E*>(pre1);
    t.u_out = static_cast<E*>(pre3);
    if constexpr (sizeof(E) == 4) return launch_ffn_gate_up_f32(f, t, workspace, st);
    else return launch_ffn_gate_up_bf16(f, t, workspace, st);
  };
  return f.dtype == MOE_F32 ? run(float{}) : run(uint16_t{});
}

hipError_t launch_ffn_backward(const moe_ffn_t& f, const void* dy, const int32_t* offsets, const void* x,
                               const void* pre1, const void* pre3, const void* h, const void* w1, const void* w3,
                               const void* w2, void* dx, void* dw1, void* dw3, void* dw2, void* workspace,
                               hipStream_t st) {
  auto run = [&](auto e) {
    using E = decltype(e);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    FfnTensors<E> t{};
    t.offsets = offsets;
    t.dy = static_cast<const E*>(dy);
    t.x = static_cast<const E*>(x);
    t.g = static_cast<const E*>(pre1);
    t.u = static_cast<const E*>(pre3);
    t.h = static_cast<const E*>(h);
    t.w1 = static_cast<const E*>(w1);
    t.w3 = static_cast<const E*>(w3);
    t.w2 = static_cast<const E*>(w2);
    t.dx = static_cast<E*>(dx);
    t.dw1 = static_cast<E*>(dw1);
    t.dw3 = static_cast<E*>(dw3);
    t.dw2 = static_cast<E*>(dw2);
    t.dg = reinterpret_cast<E*>(ws);
    t.du = reinterpret_cast<E*>(ws + pre_bytes(f));
    void* partials = ws + 2 * pre_bytes(f);
    if constexpr (sizeof(E) == 4) return launch_ffn_backward_f32(f, t, partials, st);
    else return launch_ffn_backward_bf16(f, t, partials, st);
  };
  return f.dtype == MOE_F32 ? run(float{}) : run(uint16_t{});
}

}  // namespace moe
