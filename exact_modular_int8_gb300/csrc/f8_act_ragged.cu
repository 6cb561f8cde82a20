// f8_act_ragged.cu -- the CTA-pair product with an epilogue for rows that start or
// end off 16-byte boundaries, compiled beside the instances for those that do not.
#include "f8_pair.cuh"

namespace rg {

const void* pair_act_ragged_kernel(int act, bool residual) { return pair_act_instance<true>(act, residual); }

}  // namespace rg
