// f8_act.cu -- the CTA-pair product with an epilogue, an instance for each
// activation: a unit of its own, so that they compile beside the other products.
#include "f8_pair.cuh"

namespace rg {

namespace {
template <int ACT>
const void* address() {
  return reinterpret_cast<const void*>(f8_gemm_pair_kernel<true, true, WALK_WHOLE, ACT>);
}
}  // namespace

const void* pair_act_kernel(int act) {
  switch (act) {
    case RG_ACT_SILU: return address<RG_ACT_SILU>();
    case RG_ACT_GELU: return address<RG_ACT_GELU>();
    case RG_ACT_GELU_TANH: return address<RG_ACT_GELU_TANH>();
    default: return address<SIMPLE_ACT>();
  }
}

}  // namespace rg
