// Dense product with bias, activation and residual in its epilogue (bf16
// operands, fp32 accumulation on the matrix cores).
//
// Pages: "Mixtral" study notes, nn.Linear of MixtralMoE (the router) and of
// the projections around the experts.
//
//   y = act(x w^T + bias) + residual
//
// Up to kLinearDecodeRows rows stream the weights (linear_decode.hip); more run
// as tiles (linear_tiles.hpp).
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
#include "linear_plan.hpp"

namespace moe {

size_t linear_workspace_bytes(const moe_linear_t& l) { 
  return l.M <= kLinearDecodeRows ? 0 : product_workspace(l.M, l.N, l.K, 0);
}

hipError_t launch_linear(const moe_linear_t& l, const uint16_t* x, const uint16_t* w, const float* bias,
                         const void* residual, void* y, uint16_t* pre, void* workspace, hipStream_t st) {
  const Epilogue ep{bias, residual, y, pre, l.y_dtype == MOE_F32};
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
