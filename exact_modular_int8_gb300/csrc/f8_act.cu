// f8_act.cu -- the CTA-pair product with an epilogue, an instance for each
// activation: a unit of its own, so that they compile beside the other products.
#include "f8_pair.cuh"

namespace rg {

namespace {
template <int ACT>
const void* address(bool residual) {
  return residual ? reinterpret_cast<const void*>(f8_gemm_pair_kernel<true, true, WALK_WHOLE, ACT, true>)
                  : reinterpret_cast<const void*>(f8_gemm_pair_kernel<true, true, WALK_WHOLE, ACT, false>);
}
}  // namespace

const void* pair_act_kernel(int act, bool residual) {
  switch (act) {
    case RG_ACT_SILU: return address<RG_ACT_SILU>(residual);
    case RG_ACT_GELU: return address<RG_ACT_GELU>(residual);
    case RG_ACT_GELU_TANH: return address<RG_ACT_GELU_TANH>(residual);
    default: return address<SIMPLE_ACT>(residual);
  }
}

}  // namespace rg
