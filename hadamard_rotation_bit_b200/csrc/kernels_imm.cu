// Instantiations of the int8 matrix product and their lookup.
#include "hadq_launch.h"
#include "hadq_imm.cuh"

namespace hadq {
namespace launch {

ImmFn imm_plain_for(bool out_bf16) {
  return out_bf16 ? &imm::imm_plain_kernel<true> : &imm::imm_plain_kernel<false>;
}

}  // namespace launch
}  // namespace hadq
