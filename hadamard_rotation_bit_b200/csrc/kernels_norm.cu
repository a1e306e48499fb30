// Instantiations of the norm kernels and their lookup; this unit owns a fault
// word of its own (hadq_tc_fault).
#include "hadq_launch.h"
#include "hadq_norm.cuh"

namespace hadq {
namespace launch {
namespace {

template <bool BF16, bool RES>
NormVariant pick(int64_t rows, int64_t n) {
  const int64_t chunks = n / 8;
  auto v = [](auto fn, int threads, int rpc) { return NormVariant{fn, threads * rpc, rpc}; };
  if (chunks <= 32) return v(&norm::rmsnorm_quant_kernel<BF16, RES, 32, 4, 1>, 32, 4);
  if (chunks <= 64) return v(&norm::rmsnorm_quant_kernel<BF16, RES, 32, 4, 2>, 32, 4);
  if (chunks <= 128) return v(&norm::rmsnorm_quant_kernel<BF16, RES, 128, 1, 1>, 128, 1);
  if (chunks <= 256) return v(&norm::rmsnorm_quant_kernel<BF16, RES, 128, 1, 2>, 128, 1);
  if (chunks <= 512) return v(&norm::rmsnorm_quant_kernel<BF16, RES, 256, 1, 2>, 256, 1);
  if (chunks <= 1024) return v(&norm::rmsnorm_quant_kernel<BF16, RES, 512, 1, 2>, 512, 1);
  if (chunks <= 2048) return v(&norm::rmsnorm_quant_kernel<BF16, RES, 512, 1, 4>, 512, 1);
  return v(&norm::rmsnorm_quant_kernel<BF16, RES, 1024, 1, 4>, 1024, 1);
}

template <bool BF16, bool RES>
NormRingVariant pick_ring(int64_t n) {
  const int64_t chunks = n / 8;
  if (chunks <= 512) return NormRingVariant{&norm::rmsnorm_ring_kernel<BF16, RES, 256, 2>, 256};
  if (chunks <= 1024) return NormRingVariant{&norm::rmsnorm_ring_kernel<BF16, RES, 256, 4>, 256};
  return NormRingVariant{&norm::rmsnorm_ring_kernel<BF16, RES, 512, 4>, 512};
}

}  // namespace

NormRingVariant norm_ring_for(bool bf16, bool residual, int64_t n) {
  if (bf16) return residual ? pick_ring<true, true>(n) : pick_ring<true, false>(n);
  return residual ? pick_ring<false, true>(n) : pick_ring<false, false>(n);
}

int norm_fault_bits(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, tc::hadq_tc_fault, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(tc::hadq_tc_fault, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return static_cast<int>(v);
}

NormVariant norm_kernel_for(bool bf16, bool residual, int64_t rows, int64_t n) {
  if (bf16) return residual ? pick<true, true>(rows, n) : pick<true, false>(rows, n);
  return residual ? pick<false, true>(rows, n) : pick<false, false>(rows, n);
}

}  // namespace launch
}  // namespace hadq
