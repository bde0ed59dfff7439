// Dense product with bias, activation and residual in its epilogue (fp32
// accumulation on the matrix cores).
//
// Pages: "Mixtral" study notes, nn.Linear of MixtralMoE (the router) and of
// the projections around the experts.
//
//   y = act(x w^T + bias) + residual
//
// bf16: up to kLinearDecodeRows rows stream the weights (linear_decode.hip); more
// run as tiles (linear_tiles.hpp).  fp32: linear_f32.hip.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
#include "linear_plan.hpp"

namespace moe {

size_t linear_workspace_bytes(const moe_linear_t& l) {
  if (l.dtype == MOE_F32) return linear_workspace_bytes_f32(l);
  return l.M <= kLinearDecodeRows ? 0 : product_workspace(l.M, l.N, l.K, 0);
}

hipError_t launch_linear(const moe_linear_t& l, const void* x_, const void* w_, const float* bias,
                         const void* residual, void* y, void* pre, void* workspace, hipStream_t st) {
  if (l.dtype == MOE_F32)
    return launch_linear_f32(l, static_cast<const float*>(x_), static_cast<const float*>(w_), bias,
                             static_cast<const float*>(residual), static_cast<float*>(y), static_cast<float*>(pre),
                             workspace, st);
  const uint16_t *x = static_cast<const uint16_t*>(x_), *w = static_cast<const uint16_t*>(w_);
  const Epilogue ep{bias, residual, y, static_cast<uint16_t*>(pre), l.y_dtype == MOE_F32};
  if (l.M <= kLinearDecodeRows) return launch_linear_decode(l, x, w, ep, st);
  auto run = [&](auto act) {
    return launch_product<false, false, decltype(act)::value>(x, l.K, w, l.K, l.M, l.N, l.K, workspace, ep, st);
  };
  switch (l.act) {
    case MOE_ACT_RELU: return run(std::integral_constant<int, MOE_ACT_RELU>{});
    case MOE_ACT_SILU: return run(std::integral_constant<int, MOE_ACT_SILU>{});
    case MOE_ACT_GELU: return run(std::integral_constant<int, MOE_ACT_GELU>{});
    case MOE_ACT_GELU_TANH: return run(std::integral_constant<int, MOE_ACT_GELU_TANH>{});
    default: return run(std::integral_constant<int, MOE_ACT_NONE>{});
  }
}

}  // namespace moe
