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
  return ImmSplitVariant{out_bf16 ? &imm::imm_split_kernel<C, true> : &imm::imm_split_kernel<C, false>, C::THREADS, C::SMEM_BYTES, TN, C::CTAS};
}

}  // namespace

ImmRowFn imm_row_for(int64_t m, bool out_bf16) {
  if (m == 1) return out_bf16 ? &imm::imm_row_kernel<1, true> : &imm::imm_row_kernel<1, false>;
  if (m == 2) return out_bf16 ? &imm::imm_row_kernel<2, true> : &imm::imm_row_kernel<2, false>;
  return out_bf16 ? &imm::imm_row_kernel<4, true> : &imm::imm_row_kernel<4, false>;
}

namespace {

template <int MT>
ImmWarpVariant warp_variant(int64_t m, bool out_bf16) {
  auto v = [&](auto bf16, auto f32, int nt) { return ImmWarpVariant{out_bf16 ? bf16 : f32, 16 * MT, 8 * nt}; };
  if (m <= 8) return v(&imm::imm_warp_kernel<MT, 1, true>, &imm::imm_warp_kernel<MT, 1, false>, 1);
  return v(&imm::imm_warp_kernel<MT, 2, true>, &imm::imm_warp_kernel<MT, 2, false>, 2);
}

}  // namespace

ImmWarpVariant imm_warp_for(int64_t m, bool two, bool out_bf16) {
  return two ? warp_variant<2>(m, out_bf16) : warp_variant<1>(m, out_bf16);
}

ImmSplitVariant imm_split_for(int64_t m, bool half, bool out_bf16) {
  if (m <= 32) return split<32, 4>(out_bf16);
  if (half) return split<64, 3>(out_bf16);
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
