// Instantiations of the int8 matrix product and their lookup; this unit owns a
// fault word of its own (hadq_tc_fault).
#include "hadq_launch.h"
#include "hadq_imm.cuh"

namespace hadq {
namespace launch {
namespace {

template <int TN, int STAGES>
ImmSplitVariant split(bool out_bf16) {
  using C = imm::SplitCfg<TN, STAGES>;
  return ImmSplitVariant{out_bf16 ? &imm::imm_split_kernel<C, true> : &imm::imm_split_kernel<C, false>, C::THREADS, C::SMEM_BYTES, TN};
}

}  // namespace

ImmRowFn imm_row_for(int64_t m, bool out_bf16) {
  if (m == 1) return out_bf16 ? &imm::imm_row_kernel<1, true> : &imm::imm_row_kernel<1, false>;
  if (m == 2) return out_bf16 ? &imm::imm_row_kernel<2, true> : &imm::imm_row_kernel<2, false>;
  return out_bf16 ? &imm::imm_row_kernel<4, true> : &imm::imm_row_kernel<4, false>;
}

ImmSplitVariant imm_split_for(int64_t m, bool out_bf16) {
  if (m <= 16) return split<16, 5>(out_bf16);
  if (m <= 32) return split<32, 4>(out_bf16);
  if (m <= 64) return split<64, 6>(out_bf16);
  return split<128, 4>(out_bf16);
}

ImmPairVariant imm_pair_for(bool out_bf16) {
  using C = imm::PairCfg;
  return ImmPairVariant{out_bf16 ? &imm::imm_pair_kernel<true> : &imm::imm_pair_kernel<false>, C::THREADS, C::SMEM_BYTES};
}

int imm_fault_bits(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, tc::hadq_tc_fault, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(tc::hadq_tc_fault, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return static_cast<int>(v);
}

}  // namespace launch
}  // namespace hadq
