// f8_act.cu -- the CTA-pair product with an epilogue, an instance for each
// activation: a unit of its own, so that they compile beside the other products.
#include "f8_pair.cuh"

namespace rg {

const void* pair_act_kernel(int act, bool residual) { return pair_act_instance<false>(act, residual); }

}  // namespace rg
